// Host-side checks of the norm's, the gradient norm's and the AdamW update's
// entry points for a build whose host code is instrumented with AddressSanitizer
// and UndefinedBehaviorSanitizer. Every call returns before anything is enqueued;
// device pointers are placeholders that are never dereferenced, so the program
// refuses to run where a GPU is visible. Exit status 0 when every status code is
// the expected one.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <vector>

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

int main() {
  int ndev = 0;
  if (hipGetDeviceCount(&ndev) == hipSuccess && ndev > 0) {
    printf("a GPU is visible: the host-only checks do not run here\n");
    return 0;
  }
  char* const A = reinterpret_cast<char*>(uintptr_t(0x100000));
  float* const F = reinterpret_cast<float*>(A);
  const size_t BIG = size_t(1) << 60;
  const moe_norm_opts_t layer = {MOE_NORM_LAYER, MOE_DTYPE_F32, 1e-5f}, rms = {MOE_NORM_RMS, MOE_DTYPE_BF16, 1e-6f};

  // norm: sizes over extreme dims, every one either counted or refused
  for (int64_t T : {int64_t(-1), int64_t(0), int64_t(1), int64_t(4096), int64_t(1) << 30, int64_t(1) << 62})
    for (int64_t d : {int64_t(0), int64_t(8), int64_t(12), int64_t(7168), int64_t(16384), int64_t(16392), int64_t(1) << 40})
      for (int dt : {0, 1, 2}) {
        const moe_dims_t m = {T, d, 64, 1, 1, dt};
        const bool good = T >= 0 && T < (int64_t(1) << 31) && d >= 8 && d % 8 == 0 && d <= 16384 && dt < 2;
        const size_t n = moe_norm_backward_workspace_bytes(&m, &layer);
        if ((n > 0) != good || n > (size_t(1) << 32)) {
          fprintf(stderr, "norm workspace of %lld x %lld: %zu\n", (long long)T, (long long)d, n);
          ++failures;
        }
      }
  const moe_dims_t dm = {64, 128, 64, 8, 2, MOE_DTYPE_BF16}, none = {0, 128, 64, 8, 2, MOE_DTYPE_BF16};
  EXPECT(moe_norm_forward(nullptr, &layer, A, A, A, A, A, A + 1024, F, F, nullptr), MOE_ERR_INVALID);
  EXPECT(moe_norm_forward(&dm, nullptr, A, A, A, A, A, A + 1024, F, F, nullptr), MOE_ERR_INVALID);
  EXPECT(moe_norm_forward(&dm, &rms, A, A, A, A, A, A + 1024, nullptr, F, nullptr), MOE_ERR_INVALID);
  EXPECT(moe_norm_forward(&dm, &layer, A, A, A, A, A, A, F, F, nullptr), MOE_ERR_INVALID);
  EXPECT(moe_norm_forward(&none, &layer, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr),
         MOE_OK);
  EXPECT(moe_norm_backward(&dm, &layer, A, A, A, F, F, A, A, F, F, A, 16, nullptr), MOE_ERR_WORKSPACE);
  EXPECT(moe_norm_backward(&dm, &layer, A, A, A, nullptr, F, A, A, F, F, A, BIG, nullptr), MOE_ERR_INVALID);
  EXPECT(moe_norm_backward(&dm, &rms, A, A, A, nullptr, F, A, A, F, F, A, BIG, nullptr), MOE_ERR_INVALID);

  // lists: long ones, sizes up to the limits and past them
  std::vector<moe_grad_t> g(5000, moe_grad_t{A, 8193, MOE_DTYPE_BF16});
  EXPECT(moe_grad_norm_workspace_bytes(g.data(), 5000) > 0, true);
  for (auto& e : g) e.n = int64_t(1) << 36;
  EXPECT(moe_grad_norm_workspace_bytes(g.data(), 5000) > 0, true);
  EXPECT(moe_grad_norm(g.data(), 5000, 1.0, 1.0, F, A, 64, nullptr), MOE_ERR_WORKSPACE);
  g[4999].n = (int64_t(1) << 36) + 1;
  EXPECT(moe_grad_norm_workspace_bytes(g.data(), 5000), 0);
  EXPECT(moe_grad_norm(g.data(), 5000, 1.0, 1.0, F, A, BIG, nullptr), MOE_ERR_UNSUPPORTED);
  g[4999].n = INT64_MAX;
  EXPECT(moe_grad_norm(g.data(), 5000, 1.0, 1.0, F, A, BIG, nullptr), MOE_ERR_UNSUPPORTED);
  g[4999].n = INT64_MIN;
  EXPECT(moe_grad_norm(g.data(), 5000, 1.0, 1.0, F, A, BIG, nullptr), MOE_ERR_INVALID);
  EXPECT(moe_grad_norm(nullptr, 1, 1.0, 1.0, F, A, BIG, nullptr), MOE_ERR_INVALID);
  EXPECT(moe_grad_norm(g.data(), INT32_MIN, 1.0, 1.0, F, A, BIG, nullptr), MOE_ERR_INVALID);
  EXPECT(moe_grad_norm(g.data(), INT32_MAX, 1.0, 1.0, F, A, BIG, nullptr), MOE_ERR_UNSUPPORTED);
  EXPECT(moe_grad_norm(g.data(), 1, NAN, 1.0, F, A, BIG, nullptr), MOE_ERR_INVALID);

  // the update: thousands of tensors of which the last repeats a buffer of the first
  const int n = 3000;
  std::vector<moe_adam_tensor_t> t(n);
  for (int i = 0; i < n; ++i) {
    char* p = A + int64_t(i) * 4096;
    t[i] = {p, nullptr, p + 512, p + 1024, reinterpret_cast<uint8_t*>(p + 1536), reinterpret_cast<uint8_t*>(p + 1600), 64,
            MOE_DTYPE_BF16};
    g[i] = {p + 2048, 64, MOE_DTYPE_F32};
  }
  const moe_adam_opts_t o32 = {1e-3, 0.9, 0.999, 1e-8, 0.1, INT64_MAX, 32, 0}, o8 = {1e-3, 0.9, 0.999, 1e-8, 0.1, 1, 8, 0};
  const uint64_t* const R = reinterpret_cast<const uint64_t*>(A);
  t[n - 1].v = t[0].m;
  EXPECT(moe_adam_step(&o32, t.data(), g.data(), n, nullptr, nullptr, nullptr, nullptr), MOE_ERR_INVALID);
  t[n - 1].v = A + (int64_t(1) << 30);
  t[n - 1].m_scale = t[5].v_scale;
  EXPECT(moe_adam_step(&o8, t.data(), g.data(), n, nullptr, nullptr, R, nullptr), MOE_ERR_INVALID);
  EXPECT(moe_adam_step(&o8, t.data(), g.data(), n, nullptr, nullptr, nullptr, nullptr), MOE_ERR_INVALID);
  g[7].grad = t[9].param;
  EXPECT(moe_adam_step(&o32, t.data(), g.data(), n, nullptr, nullptr, nullptr, nullptr), MOE_ERR_INVALID);
  g[7].n = 65;
  EXPECT(moe_adam_step(&o32, t.data(), g.data(), n, nullptr, nullptr, nullptr, nullptr), MOE_ERR_INVALID);
  t[7].n = INT64_MAX;
  EXPECT(moe_adam_step(&o32, t.data(), g.data(), n, nullptr, nullptr, nullptr, nullptr), MOE_ERR_UNSUPPORTED);
  t[7].n = INT64_MIN;
  EXPECT(moe_adam_step(&o32, t.data(), g.data(), n, nullptr, nullptr, nullptr, nullptr), MOE_ERR_INVALID);
  EXPECT(moe_adam_step(&o32, t.data(), g.data(), 0, nullptr, nullptr, nullptr, nullptr), MOE_OK);
  EXPECT(moe_adam_step(nullptr, t.data(), g.data(), 1, nullptr, nullptr, nullptr, nullptr), MOE_ERR_INVALID);
  EXPECT(moe_adam_step(&o32, t.data(), g.data(), INT32_MAX, nullptr, nullptr, nullptr, nullptr), MOE_ERR_UNSUPPORTED);
  std::vector<void*> out(n, A);
  out[n - 1] = nullptr;
  t[7].n = 64;
  EXPECT(moe_adam_state_values(t.data(), n, out.data(), out.data(), MOE_DTYPE_BF16, nullptr), MOE_ERR_INVALID);
  EXPECT(moe_adam_state_values(t.data(), -1, out.data(), out.data(), MOE_DTYPE_BF16, nullptr), MOE_ERR_INVALID);
  EXPECT(moe_adam_state_values(t.data(), 0, nullptr, nullptr, MOE_DTYPE_BF16, nullptr), MOE_OK);
  if (failures) fprintf(stderr, "%d checks failed\n", failures);
  return failures ? 1 : 0;
}

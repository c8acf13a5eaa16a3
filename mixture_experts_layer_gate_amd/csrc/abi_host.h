// Host-side helpers shared by the files that define C entry points: argument
// checks, workspace carving and stage timing (internal to the library).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <mutex>
#include <vector>

#include "moe.h"

namespace moe {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

// ---------------- stage timing (one process-wide record, in moe_abi.hip) ----------------
struct Timing {
  std::mutex mu;
  bool on = false;
  int cap = 0;
  unsigned mask = 0xffffffffu;
  std::vector<hipEvent_t> ev[MOE_NUM_STAGES][2];
  int n[MOE_NUM_STAGES] = {0};
};
extern Timing g_timing;

struct StageScope {
  int stage;
  hipStream_t s;
  int slot = -1;
  StageScope(int st, hipStream_t stream) : stage(st), s(stream) {
    if (!g_timing.on || !((g_timing.mask >> stage) & 1u)) return;
    if (g_timing.n[stage] < g_timing.cap) {
      slot = g_timing.n[stage]++;
      (void)hipEventRecord(g_timing.ev[stage][0][slot], s);
    }
  }
  ~StageScope() {
    if (slot >= 0) (void)hipEventRecord(g_timing.ev[stage][1][slot], s);
  }
};

// ---------------- validation ----------------
// a * b * c < lim, computed without overflow (a, b, c >= 0)
inline bool product_below(int64_t a, int64_t b, int64_t c, int64_t lim) {
  return static_cast<__int128>(a) * b * c < static_cast<__int128>(lim);
}

inline int check_dims(const moe_dims_t* dm) {
  if (!dm) return MOE_ERR_INVALID;
  if (dm->T < 0 || dm->d < 1 || dm->f < 1) return MOE_ERR_INVALID;
  if (dm->d >= (int64_t(1) << 31) || dm->f >= (int64_t(1) << 31)) return MOE_ERR_INVALID;
  if (dm->k < 1 || dm->E < dm->k || dm->E > 1024) return MOE_ERR_INVALID;
  if (dm->dtype != MOE_DTYPE_F32 && dm->dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID;
  // T*k and T*E below 2^31 (k, E >= 1, so T first: the products then fit in 64 bits)
  if (dm->T >= (int64_t(1) << 31)) return MOE_ERR_INVALID;
  if (dm->T * dm->k >= (int64_t(1) << 31) || dm->T * dm->E >= (int64_t(1) << 31)) return MOE_ERR_INVALID;
  // every workspace piece ([T*k][max(d, f)] fp32 at most, and the backward's
  // transposed activations) stays far inside size_t
  const int64_t wide = dm->d > dm->f ? dm->d : dm->f;
  if (!product_below(dm->T * dm->k + 64 * int64_t(dm->E) + 64, 2 * wide, 8, int64_t(1) << 60)) return MOE_ERR_INVALID;
  return MOE_OK;
}

inline bool ok16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline bool ok8(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 7) == 0; }
inline bool ok4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
inline bool ok4_or_null(const void* p) { return !p || (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// ---------------- workspace layouts ----------------
struct Carver {
  char* base;
  size_t off = 0;
  explicit Carver(void* b) : base(static_cast<char*>(b)) {}
  template <typename P>
  P* take(size_t bytes) {
    P* p = base ? reinterpret_cast<P*>(base + off) : nullptr;
    off = align_up(off + bytes);
    return p;
  }
};

inline int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

}  // namespace moe
